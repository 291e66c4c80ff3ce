"""The gated delta rule at sizes that leave parts of the kernels' tiles empty: 64 < N < 128 with
a wave split at the last key number, P off the 16 channels of a wave, a row's end and the
sequence's end inside a chunk, every pair of input and output types; and fp32 results at a bar
that a lost part of an operand would not pass.

Bars, relative L2.  fp32 outputs: a result passes through five products (K S, T R, U K of the state; Q S and the
query matrix times U, or their like in the gradients).  Each rounds its operands' parts and its
accumulator about a dozen times, by at most 2^-24 each and 2^-24 / sqrt(3) in the root mean square:
2^-24 sqrt(12 / 3 * 5) = 4.5 * 2^-24, and what the state carries over from earlier chunks adds
about as much again in quadrature, 6.3 * 2^-24 = 3.8e-7.  The bar is three times that, 1.2e-6 (20 *
2^-24).  With two parts of three, numbers are off by up to 2^-17, 2^-17 / sqrt(12) = 2.2e-6 in the root mean
square (test_two_parts_would_not_pass, on the oracle).  dA and ddelta_bias are sums that cancel
to a few percent of their terms and keep the bar of test_gdr_bwd_gpu.py, 4e-5.
bf16 outputs: round(x + d) is no farther from x + d than round(x), so it is off by at most
|round(x) - x| + 2 |d|: the bar is the rounding of the reference itself plus twice what d may
be, the fp32 bar, or 2^-16 for y, whose products leave out parts of 2^-17 and 2^-18 of their terms."""
import numpy as np
import pytest

from helpers import bf16_floor, f64, from_dev, log, rel_l2, to_dev
from oracle import gdr as O
from selective_state_space_75_amd import workloads as W

BAR = 20 * 2.0 ** -24
SUM_BAR = 4e-5
NAMES = ("q", "k", "v", "delta_raw", "beta_raw", "A", "delta_bias")


def _parts(x, n):
    """x as the sum of n bf16 numbers, each rounded to nearest."""
    out = np.zeros_like(x)
    for _ in range(n):
        out += f64(W.f32_to_bf16_bits((x - out).astype(np.float32)))
    return out


def test_two_parts_would_not_pass():
    x = W.gdr_inputs(1, 2, 1, 40, 72, 70, "f32", 8100)
    _, S = O.gdr(*[f64(x[n]) for n in NAMES], groups=1, norm=True)
    S = f64(S.astype(np.float32)).reshape(2, 40, 72)
    q = f64(x["q"])[0, :, -1]
    want = S @ q
    assert rel_l2(_parts(S, 3) @ q, want) < BAR / 10
    assert rel_l2(_parts(S, 2) @ q, want) > BAR


CASES = [
    # B, H, G, P, N, L, lengths: waves split at N (72 = 4 * 16 + 8, 100 = 6 * 16 + 4, 41), at P
    (2, 2, 1, 40, 72, 75, [75, 33]),
    (1, 3, 1, 72, 100, 101, None),
    (2, 2, 2, 17, 128, 97, [64, 90]),
    (1, 2, 1, 130, 41, 130, None),
]


def _inputs(case, dtype, dev, seed):
    B, H, G, P, N, L, lengths = case
    x = W.gdr_inputs(B, H, G, P, N, L, dtype, seed + P + N)
    ref = {n: f64(a.copy()) for n, a in x.items()}
    if lengths:
        for n in ("q", "k", "v", "delta_raw", "beta_raw", "dy"):
            for b, ln in enumerate(lengths):
                x[n][b, :, ln:] = np.uint16(0x7fc0) if x[n].dtype == np.uint16 else np.nan
    return {n: to_dev(a, dev) for n, a in x.items()}, ref


def _lengths(case, dev):
    import torch
    return None if case[6] is None else torch.tensor(case[6], dtype=torch.int32, device=dev)


def _check(got, want, what, bar=BAR):
    import torch
    if got.dtype == torch.bfloat16:
        bar = bf16_floor(want) + 2 * (2.0 ** -16 if what == "y" else bar)
    e = rel_l2(from_dev(got), want)
    log("  %s: rel_l2=%.3e" % (what, e))
    assert e <= bar, "%s rel L2 %.6e > %.6e" % (what, e, bar)


@pytest.mark.gpu
@pytest.mark.parametrize("kernel,segments", [("token", 0), ("chunk", 0), ("chunk", 3)])
@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("f32", "bf16"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "B%dH%dG%dP%dN%dL%d" % c[:6])
def test_forward(case, dtype, out, kernel, segments, dev):
    import torch
    import selective_state_space_75_amd as m
    B, H, G, P, N, L, lengths = case
    log("[gdr variants] %s %s to %s, %s %d" % (case, dtype, out, kernel, segments))
    t, ref = _inputs(case, dtype, dev, 8200)
    with m.gdr_test_knobs(kernel=kernel, segments=segments):
        y, S = m.gdr_fwd(*[t[n] for n in NAMES], groups=G, initial_state=t["initial_state"], lengths=_lengths(case, dev),
                         qk_norm=True, return_final_state=True,
                         out_dtype=torch.float32 if out == "f32" else torch.bfloat16)
    torch.cuda.synchronize()
    yr, Sr = O.gdr(*[ref[n] for n in NAMES], groups=G, initial_state=ref["initial_state"], lengths=lengths, norm=True)
    _check(y, yr, "y")
    _check(S, Sr, "final state")
    for b, ln in enumerate(lengths or []):
        assert not y[b, :, ln:].any()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,grad", [("f32", "f32"), ("f32", "bf16"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "B%dH%dG%dP%dN%dL%d" % c[:6])
def test_backward(case, dtype, grad, dev):
    import torch
    import selective_state_space_75_amd as m
    B, H, G, P, N, L, lengths = case
    log("[gdr variants] %s %s, gradients %s" % (case, dtype, grad))
    t, ref = _inputs(case, dtype, dev, 8300)
    dy = t["dy"].to(torch.float32 if grad == "f32" else torch.bfloat16)
    g = m.gdr_bwd(*[t[n] for n in NAMES], dy, groups=G, initial_state=t["initial_state"],
                  dfinal_state=t["dfinal_state"], lengths=_lengths(case, dev), qk_norm=True)
    torch.cuda.synchronize()
    dyr = f64(from_dev(dy))
    for b, ln in enumerate(lengths or []):
        dyr[b, :, ln:] = 0.0
    want = O.gdr_bwd(*[ref[n] for n in NAMES], dyr, groups=G, initial_state=ref["initial_state"],
                     dfinal_state=ref["dfinal_state"], lengths=lengths, norm=True)
    for n, a in g.items():
        _check(a, want[n], n, SUM_BAR if n in ("dA", "ddelta_bias") else BAR)
        if lengths and a.dim() == 3 and n != "dinitial_state":
            for b, ln in enumerate(lengths):
                assert not a[b, :, ln:].any(), n
