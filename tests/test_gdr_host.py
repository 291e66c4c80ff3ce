"""Host-side checks of the gated delta rule's and the 8-bit state cache's calls:
exported symbols, workspace sizes, and every refusal, before any HIP call (fake,
never-dereferenced addresses; no GPU needed)."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

from selective_state_space_75_amd import _lib  # noqa: E402

NULL, SHAPE, DTYPE, ALIGN, UNSUP, WS = -1, -2, -3, -4, -5, -6
F32, BF16 = 0, 1
P = 0x10000


def test_header_symbols_are_exported():
    for h in ("mamba_gdr.h", "mamba_state_cache.h"):
        src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", h), encoding="utf-8").read(), flags=re.S)
        names = set(re.findall(r"\b(mamba_[a-z0-9_]+)\s*\(", src))
        assert names
        for n in names:
            assert hasattr(_lib.lib(), n), n


def _vp(v):
    return ctypes.c_void_p(v) if v is not None else None


def fwd(**kw):
    a = dict(q=P, k=P, v=P, delta=P, beta=P, A=P, bias=None, init=None, lengths=None, y=P, fs=None, B=2, H=4, G=2,
             Pd=64, N=128, L=256, qs=None, ks=None, vs=None, ind=BF16, outd=BF16, flags=0, ws=P, wsb=1 << 40)
    a.update(kw)
    qs = a["G"] * a["N"] * a["L"]
    vs = a["H"] * a["Pd"] * a["L"]
    return _lib.lib().mamba_gdr_fwd(*[_vp(a[n]) for n in ("q", "k", "v", "delta", "beta", "A", "bias", "init",
                                                         "lengths", "y", "fs")],
                                    a["B"], a["H"], a["G"], a["Pd"], a["N"], a["L"],
                                    qs if a["qs"] is None else a["qs"], qs if a["ks"] is None else a["ks"],
                                    vs if a["vs"] is None else a["vs"], 0.5, a["ind"], a["outd"], a["flags"],
                                    _vp(a["ws"]), a["wsb"], None)


SHARED = [
    (dict(ind=7), DTYPE), (dict(outd=2), DTYPE), (dict(flags=0x1), UNSUP), (dict(flags=0x8), UNSUP),
    (dict(B=0), SHAPE), (dict(H=0), SHAPE), (dict(G=0), SHAPE), (dict(Pd=0), SHAPE), (dict(N=0), SHAPE),
    (dict(B=-1), SHAPE), (dict(H=3, G=2), SHAPE), (dict(G=8), SHAPE), (dict(N=129), UNSUP), (dict(N=256), UNSUP),
    (dict(B=1 << 30, H=1 << 20, Pd=1 << 20), SHAPE), (dict(H=1 << 40, G=1, Pd=1 << 40), SHAPE),
    (dict(qs=1), SHAPE), (dict(ks=-1), SHAPE), (dict(vs=100), SHAPE), (dict(qs=1 << 62), SHAPE),
    (dict(q=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL), (dict(delta=None), NULL),
    (dict(beta=None), NULL), (dict(A=None), NULL), (dict(y=None), NULL),
    (dict(q=P + 1), ALIGN), (dict(v=P + 1), ALIGN), (dict(beta=P + 1), ALIGN), (dict(ind=F32, k=P + 2), ALIGN),
    (dict(outd=F32, y=P + 2), ALIGN), (dict(A=P + 2), ALIGN), (dict(bias=P + 1), ALIGN),
]


@pytest.mark.parametrize("kw,code", SHARED + [
    (dict(L=0), SHAPE), (dict(L=1 << 40, B=1 << 10), SHAPE),
    (dict(init=P + 2), ALIGN), (dict(lengths=P + 2), ALIGN), (dict(fs=P + 1), ALIGN),
    (dict(ws=None), WS), (dict(wsb=1000), WS), (dict(ws=P + 16), ALIGN),
])
def test_fwd_rejects_bad_arguments(kw, code):
    assert fwd(**kw) == code


def update(**kw):
    a = dict(state=P, slots=None, q=P, k=P, v=P, delta=P, beta=P, A=P, bias=None, y=P, B=2, H=4, G=2, Pd=64, N=128,
             S=2, qs=None, ks=None, vs=None, ind=BF16, outd=BF16, flags=0)
    a.update(kw)
    qs, vs = a["G"] * a["N"], a["H"] * a["Pd"]
    return _lib.lib().mamba_gdr_update(*[_vp(a[n]) for n in ("state", "slots", "q", "k", "v", "delta", "beta", "A",
                                                            "bias", "y")],
                                       a["B"], a["H"], a["G"], a["Pd"], a["N"], a["S"],
                                       qs if a["qs"] is None else a["qs"], qs if a["ks"] is None else a["ks"],
                                       vs if a["vs"] is None else a["vs"], 0.5, a["ind"], a["outd"], a["flags"], None)


@pytest.mark.parametrize("kw,code", SHARED + [
    (dict(S=1), SHAPE), (dict(S=0, slots=P), SHAPE), (dict(S=1 << 50, slots=P), SHAPE),
    (dict(state=None), NULL), (dict(state=P + 2), ALIGN), (dict(slots=P + 2), ALIGN),
])
def test_update_rejects_bad_arguments(kw, code):
    assert update(**kw) == code


def bwd(**kw):
    names = ("q", "k", "v", "delta", "beta", "A", "bias", "init", "lengths", "dy", "dfs", "dq", "dk", "dv", "ddelta",
             "dbeta", "dA", "dbias", "dinit")
    a = dict.fromkeys(names, P)
    a.update(bias=None, init=None, lengths=None, dfs=None, dinit=None, B=2, H=4, G=2, Pd=64, N=128, L=256, qs=None,
             ks=None, vs=None, ind=BF16, outd=BF16, flags=0, ws=P, wsb=1 << 40)
    a.update(kw)
    if "y" in kw:                                     # the shared refusals speak of y: here its gradient
        a["dy"] = kw["y"]
    qs, vs = a["G"] * a["N"] * a["L"], a["H"] * a["Pd"] * a["L"]
    return _lib.lib().mamba_gdr_bwd(*[_vp(a[n]) for n in names], a["B"], a["H"], a["G"], a["Pd"], a["N"], a["L"],
                                    qs if a["qs"] is None else a["qs"], qs if a["ks"] is None else a["ks"],
                                    vs if a["vs"] is None else a["vs"], 0.5, a["ind"], a["outd"], a["flags"],
                                    _vp(a["ws"]), a["wsb"], None)


@pytest.mark.parametrize("kw,code", SHARED + [
    (dict(L=0), SHAPE), (dict(L=1 << 40, B=1 << 10), SHAPE),
    (dict(dq=None), NULL), (dict(dk=None), NULL), (dict(dv=None), NULL), (dict(ddelta=None), NULL),
    (dict(dbeta=None), NULL), (dict(dA=None), NULL), (dict(dbias=None), NULL),
    (dict(dq=P + 1), ALIGN), (dict(outd=F32, dbeta=P + 2), ALIGN), (dict(dA=P + 2), ALIGN), (dict(dinit=P + 2), ALIGN),
    (dict(dfs=P + 2), ALIGN), (dict(init=P + 1), ALIGN),
    (dict(ws=None), WS), (dict(wsb=1 << 20), WS), (dict(ws=P + 16), ALIGN),
])
def test_bwd_rejects_bad_arguments(kw, code):
    assert bwd(**kw) == code


def cache(write, **kw):
    a = dict(state=P, slots=None, codes=P, exps=P, rows=2, n=64, S=4, dt=F32)
    a.update(kw)
    L = _lib.lib()
    if write:
        return L.mamba_state_cache_write(_vp(a["state"]), _vp(a["slots"]), _vp(a["codes"]), _vp(a["exps"]), a["rows"],
                                         a["n"], a["S"], a["dt"], None)
    return L.mamba_state_cache_read(_vp(a["codes"]), _vp(a["exps"]), _vp(a["slots"]), _vp(a["state"]), a["rows"],
                                    a["n"], a["S"], a["dt"], None)


@pytest.mark.parametrize("write", [True, False])
@pytest.mark.parametrize("kw,code", [
    (dict(dt=5), DTYPE), (dict(rows=0), SHAPE), (dict(n=0), SHAPE), (dict(n=-4), SHAPE), (dict(S=0), SHAPE),
    (dict(S=1), SHAPE), (dict(rows=1 << 40, n=1 << 20, S=1 << 40), SHAPE), (dict(rows=1 << 40, n=1, slots=P), SHAPE),
    (dict(state=None), NULL), (dict(codes=None), NULL), (dict(exps=None), NULL),
    (dict(state=P + 2), ALIGN), (dict(dt=BF16, state=P + 1), ALIGN), (dict(slots=P + 2), ALIGN),
])
def test_cache_rejects_bad_arguments(write, kw, code):
    assert cache(write, **kw) == code


def test_workspace_size_of_invalid_shapes():
    bad = ctypes.c_size_t(-1).value
    ws = _lib.lib().mamba_gdr_workspace_size
    assert ws(2, 3, 2, 64, 128, 256, BF16) == bad
    assert ws(2, 4, 2, 64, 129, 256, BF16) == bad
    assert ws(0, 4, 2, 64, 128, 256, BF16) == bad
    assert ws(2, 4, 2, 64, 128, 256, 9) == bad
    assert ws(2, 4, 2, 64, 128, 256, BF16) < bad
    with pytest.raises(_lib.MambaError):
        _lib.gdr_workspace_size(2, 3, 2, 64, 128, 256)


def test_workspace_size_plan():
    """6 operand planes of 2 KB and 512 bytes of factors per head and chunk of 32 tokens; a partial last chunk
    of k, q and v per row; few heads over a long L add segments: a transition and an end state for each but
    the last, a start for each."""
    ws = _lib.gdr_workspace_size
    a = lambda x: (x + 255) // 256 * 256  # noqa: E731
    assert ws(4, 40, 20, 128, 128, 1) == 0
    blocks = 4 * 40 * 64
    assert ws(4, 40, 20, 128, 128, 2048) == (a(blocks * 6 * 2048) + a(blocks * 512) + 2 * a(80 * 128 * 64)
                                             + a(160 * 128 * 64))
    with _lib.gdr_test_knobs(kernel="chunk", segments=3):
        blocks = 2 * 4
        assert ws(1, 2, 2, 40, 96, 100) == (a(blocks * 6 * 2048) + a(blocks * 512) + 2 * a(2 * 96 * 64)
                                            + a(2 * 40 * 64) + a(2 * 1 * 96 * 96 * 4)
                                            + a(2 * 1 * 40 * 96 * 4) + a(2 * 2 * 40 * 96 * 4))   # 4 chunks: 2 + 2
    with _lib.gdr_test_knobs(kernel="token"):
        assert ws(4, 40, 20, 128, 128, 2048) == 0
    # backward: 9 planes and 1 KB of factors per chunk, updates and gradients of v (fp32), a state per block
    # of 4 chunks and per chunk, sums of dq and dk over value heads (P and N rounded up to 64), two sums per
    # block; one row of 2 heads, one key head, 5 chunks in 2 blocks
    bw = _lib.lib().mamba_gdr_bwd_workspace_size(1, 2, 1, 40, 96, 130, BF16, F32)
    assert bw == (a(10 * 9 * 2048) + a(10 * 1024) + 2 * a(96 * 64) + a(2 * 40 * 64) + a(2 * 40 * 128)
                  + 2 * a(10 * 64 * 128) + a(4 * 64 * 128 * 4) + a(10 * 64 * 128 * 4) + 2 * a(5 * 128 * 128) + a(4 * 8))


def test_knob_errors():
    f = _lib.lib().mamba_gdr_set_test_knobs
    assert f(3, 0) == SHAPE and f(-1, 0) == SHAPE and f(0, -1) == SHAPE
    assert f(0, 0) == 0


def test_python_binding_rejects_before_calling():
    import torch
    import selective_state_space_75_amd as m
    q = torch.zeros(2, 8, 5)
    v = torch.zeros(2, 6, 5)
    d = torch.zeros(2, 2, 5)
    A = torch.zeros(2)
    with pytest.raises(ValueError, match="GPU device"):
        m.gdr_fwd(q, q, v, d, d, A)
    with pytest.raises(ValueError, match="divide"):
        m.gdr_fwd(q, q, v, d, d, A, groups=3)
    with pytest.raises(ValueError, match="dimensions"):
        m.gdr_fwd(q[0], q, v, d, d, A)
    with pytest.raises(ValueError, match="dimensions"):
        m.gdr_update(torch.zeros(2, 6, 4), q, q, v, d, d, A)
    with pytest.raises(ValueError, match="GPU device"):
        m.state_cache_write(torch.zeros(2, 5), torch.zeros(2, 5, dtype=torch.int8), torch.zeros(2, 1, dtype=torch.uint8))
    with pytest.raises(ValueError, match="codes"):
        m.state_cache_read(torch.zeros(5, dtype=torch.int8), torch.zeros(2, 1, dtype=torch.uint8), out=torch.zeros(2, 5))


def test_a_stream_of_another_device_is_refused():
    from types import SimpleNamespace
    import torch
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        _lib._on(torch.device("cuda", 0), SimpleNamespace(device=torch.device("cuda", 1)))
