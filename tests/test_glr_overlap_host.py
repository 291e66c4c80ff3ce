"""Outputs that the caller gives must not lie over what the call reads, or over each other: workgroups read and write
in no order.  The binding's checks run here on CPU tensors, the library's entry points replaced by ones that do nothing,
so that no call of the kind ever reaches a GPU."""
import contextlib

import pytest
import torch

import selective_state_space_75_amd as m
from selective_state_space_75_amd import _lib

B, D, L, S = 2, 4, 8, 5
F32 = torch.float32


class _Nothing:
    calls = 0

    def __getattr__(self, name):
        def call(*a):
            _Nothing.calls += 1
            return 0
        return call


@pytest.fixture(autouse=True)
def on_the_host(monkeypatch):
    monkeypatch.setattr(_lib, "lib", _Nothing)
    monkeypatch.setattr(_lib, "_there", lambda dev, stream: contextlib.nullcontext())
    monkeypatch.setattr(_lib, "_raw_stream", lambda dev, stream: 0)
    monkeypatch.setattr(_lib, "_first", lambda x, dims, what: (x.device, x.dtype, _lib._dtype_code(x)))
    monkeypatch.setattr(_lib, "_workspace", lambda ws, n, dev: ws)
    _Nothing.calls = 0


def big():
    return torch.zeros(B, D, L)


def over(n, shape):
    """Tensors of n numbers in all that overlap by one number: the first `shape`, and what follows."""
    buf = torch.zeros(4096)
    k = 1
    for s in shape:
        k *= s
    return buf[:k].view(shape), buf[k - 1:k - 1 + n]


def refused(call):
    before = _Nothing.calls
    with pytest.raises(ValueError, match="overlap"):
        call()
    assert _Nothing.calls <= before + 1          # at most the workspace's size was asked for


def per(n=1):
    return -torch.ones(D)


def test_a_state_in_place_is_refused():
    h = torch.zeros(B, D)
    refused(lambda: m.glr_fwd(big(), big(), None, per(), initial_state=h, return_final_state=True, final_state=h))
    a, b = over(B * D, (B, D))
    refused(lambda: m.glr_fwd(big(), big(), None, per(), initial_state=a, return_final_state=True, final_state=b.view(B, D)))
    refused(lambda: m.glr_fwd(big(), big(), None, per(), initial_state=b.view(B, D), return_final_state=True, final_state=a))


@pytest.mark.parametrize("which", ["x", "r", "i", "z"])
def test_outputs_over_the_sequences(which):
    for out in ("y", "final_state"):
        t = {n: big() for n in ("x", "r", "i", "z")}
        a, b = over(B * D * L, (B, D, L) if out == "y" else (B, D))
        t[which] = b.view(B, D, L)
        refused(lambda: m.glr_fwd(t["x"], t["r"], t["i"], per(), z=t["z"], return_final_state=True, **{out: a}))


@pytest.mark.parametrize("which", ["A", "r_bias", "i_bias", "initial_state", "lengths", "final_state"])
def test_outputs_over_the_parameters_and_states(which):
    for out in ("y", "final_state"):
        if which == out:
            continue
        a, b = over(B * D, (B, D, L) if out == "y" else (B, D))
        kw = {"A": per(), "r_bias": per(), "i_bias": per(), "initial_state": torch.zeros(B, D), "final_state": torch.zeros(B, D),
              "lengths": torch.full((B,), L, dtype=torch.int32), out: a}
        kw[which] = b[:D] if which in ("A", "r_bias", "i_bias") else b[:B].view(torch.int32) if which == "lengths" else b.view(B, D)
        refused(lambda: m.glr_fwd(big(), big(), big(), return_final_state=True, **kw))


def one():
    return torch.zeros(B, D)


@pytest.mark.parametrize("which", ["state", "x", "r", "i", "z", "A", "r_bias", "i_bias", "slots"])
def test_a_tokens_output_over_what_it_reads(which):
    a, b = over(S * D, (B, D))
    t = {"state": torch.zeros(S, D), "x": one(), "r": one(), "i": one(), "z": one(), "A": per(), "r_bias": per(), "i_bias": per(),
         "slots": torch.zeros(B, dtype=torch.int32)}
    t[which] = (b.view(S, D) if which == "state" else b[:B].view(torch.int32) if which == "slots" else
                b[:B * D].view(B, D) if which in ("x", "r", "i", "z") else b[:D])
    refused(lambda: m.glr_update(t.pop("state"), t.pop("x"), t.pop("r"), y=a, **t))


@pytest.mark.parametrize("which", ["x", "r", "i", "z"])
def test_a_tokens_input_over_the_pool(which):
    a, b = over(B * D, (S, D))
    t = {"x": one(), "r": one(), "i": one(), "z": one()}
    t[which] = b.view(B, D)
    refused(lambda: m.glr_update(a, t["x"], t["r"], t["i"], per(), z=t["z"]))


@pytest.mark.parametrize("which", ["x", "z", "weight", "bias"])
def test_a_norms_output_over_what_it_reads(which):
    a, b = over(B * D * L, (B, D, L))
    t = {"x": big(), "z": big(), "weight": per(), "bias": per()}
    t[which] = b[:D] if which in ("weight", "bias") else b.view(B, D, L)
    refused(lambda: m.layer_norm_fwd(t["x"], t["weight"], t["bias"], t["z"], y=a))


def test_outputs_side_by_side_are_taken():
    buf = torch.zeros(4096)
    n = B * D * L
    y, x, h0, h1 = buf[:n].view(B, D, L), buf[n:2 * n].view(B, D, L), buf[2 * n:2 * n + B * D].view(B, D), \
        buf[2 * n + B * D:2 * n + 2 * B * D].view(B, D)
    A = buf[2 * n + 2 * B * D:2 * n + 2 * B * D + D]
    out = m.glr_fwd(x, x, None, A, initial_state=h0, y=y, return_final_state=True, final_state=h1)
    assert out[0] is y and out[1] is h1
    pool = buf[3 * n:3 * n + S * D].view(S, D)
    k = 3 * n + S * D
    rows = [buf[k + j * B * D:k + (j + 1) * B * D].view(B, D) for j in range(3)]
    assert m.glr_update(pool, rows[0], rows[1], None, A, y=rows[2]) is rows[2]
    assert m.layer_norm_fwd(x, A, A, y=y) is y
    wide = torch.zeros(1, 3 * D, L)
    assert m.layer_norm_fwd(wide[:, :D], y=wide[:, D:2 * D]) is not None
