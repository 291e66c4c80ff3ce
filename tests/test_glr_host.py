"""Host-side checks of the gated linear recurrence's and the layer norm's calls: exported symbols,
workspace sizes, and every refusal, before any HIP call (fake, never-dereferenced addresses; no GPU
needed)."""
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
    for h in ("mamba_glr.h", "mamba_norm.h"):
        src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", h), encoding="utf-8").read(), flags=re.S)
        names = set(re.findall(r"\b(mamba_[a-z0-9_]+)\s*\(", src))
        assert len(names) >= 3
        for n in names:
            assert hasattr(_lib.lib(), n), n


def _vp(v):
    return ctypes.c_void_p(v) if v is not None else None


def _strides(a, names, row):
    return [row if a[n] is None else a[n] for n in names]


GLR = dict(x=P, r=P, i=P, z=P, A=P, rb=None, ib=None, init=None, lengths=None, y=P, fs=None, B=2, D=6, L=256, xs=None,
           rs=None, is_=None, zs=None, ind=BF16, outd=BF16, flags=0, ws=P, wsb=1 << 40)


def fwd(**kw):
    a = {**GLR, **kw}
    return _lib.lib().mamba_glr_fwd(*[_vp(a[n]) for n in ("x", "r", "i", "z", "A", "rb", "ib", "init", "lengths", "y",
                                                         "fs")],
                                    a["B"], a["D"], a["L"], *_strides(a, ("xs", "rs", "is_", "zs"), a["D"] * a["L"]),
                                    a["ind"], a["outd"], a["flags"], _vp(a["ws"]), a["wsb"], None)


def update(**kw):
    a = {**GLR, "state": P, "slots": None, "S": 2, **kw}
    return _lib.lib().mamba_glr_update(*[_vp(a[n]) for n in ("state", "slots", "x", "r", "i", "z", "A", "rb", "ib", "y")],
                                       a["B"], a["D"], a["S"], *_strides(a, ("xs", "rs", "is_", "zs"), a["D"]), a["ind"],
                                       a["outd"], a["flags"], None)


GRADS = ("dx", "dr", "di", "dz", "dA", "drb", "dib", "dinit")


def bwd(**kw):
    a = {**GLR, **dict.fromkeys(GRADS, P), "dinit": None, "dfs": None, **kw}
    if "y" in kw:                                     # the shared refusals speak of y: here its gradient
        a["dy"] = kw["y"]
    a.setdefault("dy", P)
    return _lib.lib().mamba_glr_bwd(*[_vp(a[n]) for n in ("x", "r", "i", "z", "A", "rb", "ib", "init", "lengths", "dy",
                                                         "dfs") + GRADS],
                                    a["B"], a["D"], a["L"], *_strides(a, ("xs", "rs", "is_", "zs"), a["D"] * a["L"]),
                                    a["ind"], a["outd"], a["flags"], _vp(a["ws"]), a["wsb"], None)


SHARED = [
    (dict(ind=7), DTYPE), (dict(outd=2), DTYPE), (dict(flags=0x1), UNSUP), (dict(flags=0x4), UNSUP),
    (dict(flags=0x10), UNSUP), (dict(B=0), SHAPE), (dict(D=0), SHAPE), (dict(B=-1), SHAPE), (dict(D=-3), SHAPE),
    (dict(B=1 << 30, D=1 << 30), SHAPE), (dict(B=1 << 40, D=1 << 40), SHAPE),
    (dict(xs=1), SHAPE), (dict(rs=-1), SHAPE), (dict(is_=5), SHAPE), (dict(zs=0), SHAPE), (dict(xs=1 << 62), SHAPE),
    (dict(x=None), NULL), (dict(r=None), NULL), (dict(A=None), NULL), (dict(y=None), NULL),
    (dict(x=P + 1), ALIGN), (dict(r=P + 1), ALIGN), (dict(i=P + 1), ALIGN), (dict(z=P + 1), ALIGN),
    (dict(ind=F32, r=P + 2), ALIGN), (dict(outd=F32, y=P + 2), ALIGN), (dict(y=P + 1), ALIGN), (dict(A=P + 2), ALIGN),
    (dict(rb=P + 1), ALIGN), (dict(ib=P + 2), ALIGN),
]
SEQUENCES = [(dict(L=0), SHAPE), (dict(L=1 << 45), SHAPE), (dict(B=1 << 13, D=1 << 14, L=1), SHAPE),
             (dict(init=P + 2), ALIGN), (dict(lengths=P + 2), ALIGN)]


@pytest.mark.parametrize("kw,code", SHARED + SEQUENCES + [
    (dict(fs=P + 1), ALIGN), (dict(B=1, D=2, L=1 << 20, ws=None), WS), (dict(B=1, D=2, L=1 << 20, wsb=7), WS),
    (dict(B=1, D=2, L=1 << 20, ws=P + 16), ALIGN),
])
def test_fwd_rejects_bad_arguments(kw, code):
    assert fwd(**kw) == code


@pytest.mark.parametrize("kw,code", SHARED + [
    (dict(S=1), SHAPE), (dict(S=0, slots=P), SHAPE), (dict(S=1 << 50, slots=P), SHAPE), (dict(B=1 << 25, S=1 << 25), SHAPE),
    (dict(state=None), NULL), (dict(state=P + 2), ALIGN), (dict(slots=P + 2), ALIGN),
])
def test_update_rejects_bad_arguments(kw, code):
    assert update(**kw) == code


@pytest.mark.parametrize("kw,code", SHARED + SEQUENCES + [
    (dict(dx=None), NULL), (dict(dr=None), NULL), (dict(di=None), NULL), (dict(dz=None), NULL), (dict(dA=None), NULL),
    (dict(drb=None), NULL), (dict(dib=None), NULL), (dict(dx=P + 1), ALIGN), (dict(outd=F32, dz=P + 2), ALIGN),
    (dict(dA=P + 2), ALIGN), (dict(dib=P + 2), ALIGN), (dict(dinit=P + 2), ALIGN), (dict(dfs=P + 2), ALIGN),
    (dict(ws=None), WS), (dict(wsb=100), WS), (dict(ws=P + 16), ALIGN),
])
def test_bwd_rejects_bad_arguments(kw, code):
    assert bwd(**kw) == code


NORM = dict(x=P, z=P, w=P, b=P, y=P, dy=P, dx=P, dz=P, dw=P, db=P, B=2, D=12, L=40, G=3, xs=None, zs=None, eps=1e-5, ind=BF16,
            outd=BF16, flags=0, ws=P, wsb=1 << 40)


def norm_fwd(**kw):
    a = {**NORM, **kw}
    return _lib.lib().mamba_layer_norm_fwd(*[_vp(a[n]) for n in ("x", "z", "w", "b", "y")], a["B"], a["D"], a["L"], a["G"],
                                           *_strides(a, ("xs", "zs"), a["D"] * a["L"]), a["eps"], a["ind"], a["outd"],
                                           a["flags"], _vp(a["ws"]), a["wsb"], None)


def norm_bwd(**kw):
    a = {**NORM, **kw}
    if "y" in kw:
        a["dy"] = kw["y"]
    return _lib.lib().mamba_layer_norm_bwd(*[_vp(a[n]) for n in ("x", "z", "w", "b", "dy", "dx", "dz", "dw", "db")],
                                           a["B"], a["D"], a["L"], a["G"], *_strides(a, ("xs", "zs"), a["D"] * a["L"]),
                                           a["eps"], a["ind"], a["outd"], a["flags"], _vp(a["ws"]), a["wsb"], None)


NORM_SHARED = [
    (dict(ind=7), DTYPE), (dict(outd=-1), DTYPE), (dict(flags=0x8), UNSUP), (dict(eps=-1.0), UNSUP),
    (dict(eps=float("nan")), UNSUP), (dict(B=0), SHAPE), (dict(D=0), SHAPE), (dict(L=0), SHAPE), (dict(G=0), SHAPE),
    (dict(G=5), SHAPE), (dict(G=-3), SHAPE), (dict(G=24), SHAPE), (dict(L=1 << 45), SHAPE), (dict(B=1 << 60), SHAPE),
    (dict(xs=3), SHAPE), (dict(zs=-1), SHAPE), (dict(x=None), NULL), (dict(y=None), NULL), (dict(x=P + 1), ALIGN),
    (dict(z=P + 1), ALIGN), (dict(w=P + 2), ALIGN), (dict(b=P + 1), ALIGN), (dict(outd=F32, y=P + 2), ALIGN),
    (dict(ind=F32, x=P + 2), ALIGN),
]


@pytest.mark.parametrize("kw,code", NORM_SHARED + [(dict(D=10000, G=1, ws=None), WS), (dict(D=10000, G=1, wsb=3), WS), (dict(D=10000, G=1, ws=P + 16), ALIGN),
                                               (dict(B=1 << 27, D=1, G=1, L=1), SHAPE), (dict(B=1 << 14, D=1 << 12, G=1 << 12, L=64), SHAPE)])
def test_norm_fwd_rejects_bad_arguments(kw, code):
    assert norm_fwd(**kw) == code


@pytest.mark.parametrize("kw,code", NORM_SHARED + [
    (dict(dx=None), NULL), (dict(dz=None), NULL), (dict(dw=None), NULL), (dict(db=None), NULL), (dict(dx=P + 1), ALIGN),
    (dict(dw=P + 2), ALIGN), (dict(ws=None), WS), (dict(wsb=1), WS), (dict(ws=P + 16), ALIGN),
])
def test_norm_bwd_rejects_bad_arguments(kw, code):
    assert norm_bwd(**kw) == code


def test_workspace_sizes():
    L = _lib.lib()
    bad = ctypes.c_size_t(-1).value
    for f in (L.mamba_glr_workspace_size, L.mamba_glr_bwd_workspace_size):
        assert f(0, 1, 1) == bad and f(1, -1, 1) == bad and f(1 << 20, 1 << 20, 1 << 20) == bad
    assert L.mamba_glr_workspace_size(4, 5120, 2048) == 0             # rows enough: one launch
    assert 0 < L.mamba_glr_workspace_size(1, 2, 1 << 20) < 1 << 20
    assert L.mamba_glr_bwd_workspace_size(4, 5120, 2048) >= 3 * 4 * 5120 * 4
    for f in (L.mamba_layer_norm_workspace_size, L.mamba_layer_norm_bwd_workspace_size):
        assert f(2, 12, 40, 5) == bad and f(2, 12, 40, 0) == bad and f(0, 12, 40, 3) == bad
    assert L.mamba_layer_norm_workspace_size(2, 12, 40, 3) == 0 and L.mamba_layer_norm_workspace_size(128, 5120, 1, 1) == 0
    assert L.mamba_layer_norm_workspace_size(1, 10000, 64, 1) >= 2 * 64 * 4
    assert L.mamba_layer_norm_bwd_workspace_size(2, 12, 40, 3) >= 2 * 12 * 4


def test_knobs():
    L = _lib.lib()
    for waves, seg in ((-1, 0), (17, 0), (0, -1)):
        assert L.mamba_glr_set_test_knobs(waves, seg) == SHAPE
    import selective_state_space_75_amd as m
    plain = m.glr_bwd_workspace_size(1, 2, 100)
    with m.glr_test_knobs(segments=4):
        assert m.glr_bwd_workspace_size(1, 2, 100) > plain
    assert m.glr_bwd_workspace_size(1, 2, 100) == plain


def test_binding_refuses_by_name():
    import torch
    import selective_state_space_75_amd as m
    x = torch.zeros(2, 4, 8)
    with pytest.raises(ValueError, match="GPU device"):
        m.glr_fwd(x, x, None, torch.zeros(4))
    with pytest.raises(ValueError, match="GPU device"):
        m.layer_norm_bwd(x, None, None, None, x)
    with pytest.raises(TypeError, match="x must be"):
        m.glr_fwd([1.0], x)
    with pytest.raises(ValueError, match="x must be"):
        m.glr_update(x, x, x)
    with pytest.raises(ValueError, match="x must be"):
        m.layer_norm_fwd(x[0, 0])
    with pytest.raises(m.MambaError):
        m.glr_workspace_size(0, 1, 1)
    with pytest.raises(m.MambaError):
        m.glr_bwd_workspace_size(1, 1, -1)
    with pytest.raises(m.MambaError):
        m.layer_norm_bwd_workspace_size(1, 10, 1, 3)
