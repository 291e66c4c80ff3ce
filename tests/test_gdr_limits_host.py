"""Sizes whose launch would hold 2^32 threads or more are refused as a shape, before any HIP call;
one step below they pass that check and are refused for another reason (a misaligned or missing
array, so that nothing is launched)."""
import pytest

from test_gdr_host import ALIGN, BF16, F32, P, SHAPE, WS, bwd, cache, fwd, update

from selective_state_space_75_amd import _lib


@pytest.mark.parametrize("kw,B", [
    (dict(H=1 << 13, G=1 << 13, Pd=4, N=2), 1 << 13),             # one set of four rows per wave
    (dict(H=1 << 13, G=1, Pd=1, N=3), 1 << 13),                   # (a single row takes a set too)
    (dict(H=1 << 13, G=1 << 13, Pd=16, N=4), 1 << 13),            # four sets
    (dict(H=1 << 13, G=1 << 13, Pd=4, N=4, state=P + 4), 1 << 13),
])
def test_update(kw, B):
    assert update(B=B, S=B, v=P + 1, **kw) == SHAPE
    assert update(B=B - 1, S=B, v=P + 1, **kw) == ALIGN


def test_forward_token_by_token():
    with _lib.gdr_test_knobs(kernel="token"):
        kw = dict(H=1 << 13, G=1 << 13, Pd=4, N=2, L=1, v=P + 1)
        assert fwd(B=1 << 13, **kw) == SHAPE
        assert fwd(B=(1 << 13) - 1, **kw) == ALIGN


@pytest.mark.parametrize("kw,B,segments", [
    (dict(H=1 << 10, G=1 << 10, Pd=1, N=1, L=128), 1 << 12, 1),        # preparation: a workgroup per key head and chunk
    (dict(H=1 << 12, G=1, Pd=128, N=1, L=96), 1 << 11, 1),             # chain: per head and 64 channels
    (dict(H=1 << 9, G=1, Pd=64, N=128, L=160), 2731, 5),               # summaries: 4 segments x 3 slices x 512 heads
    (dict(H=1 << 10, G=1, Pd=128, N=65, L=64), 1 << 10, 2),            # carries: 512 threads per 16 channels
])
def test_forward_in_chunks(kw, B, segments):
    with _lib.gdr_test_knobs(kernel="chunk", segments=segments):
        assert fwd(B=B, ws=None, **kw) == SHAPE
        assert fwd(B=B - 1, ws=None, **kw) == WS


@pytest.mark.parametrize("kw,H", [
    (dict(B=4, G=1, Pd=1, N=1, L=128), 1 << 20),                       # pairs: per value head and chunk
    (dict(B=1 << 11, G=None, Pd=1, N=65, L=32), 1 << 12),              # grads: 512 threads per key head and 4 chunks
    (dict(B=4, G=1, Pd=64 * 4, N=1, L=32), 1 << 20),                   # chains
])
def test_backward(kw, H):
    def call(h):
        a = dict(kw)
        if a["G"] is None:
            a["G"] = h
        return bwd(H=h, ws=None, **a)
    assert call(H) == SHAPE
    assert call(H - 1) == WS


@pytest.mark.parametrize("write", [True, False])
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("n", [(1 << 20) - 1, 1 << 22])               # 1024 pieces of 1024, and of 4096 numbers
def test_cache(n, dt, write):
    assert cache(write, rows=1 << 14, n=n, S=1 << 14, dt=dt, slots=P + 2) == SHAPE
    assert cache(write, rows=(1 << 14) - 1, n=n, S=1 << 14, dt=dt, slots=P + 2) == ALIGN
