"""The gated linear recurrence and the layer norm on arrays of more than 2^31 numbers: what lies past 32-bit
offsets, against the oracle or the same call on that part alone."""
import numpy as np
import pytest

from helpers import from_dev
from oracle import glr as O
from test_glr_gpu import E, near

pytestmark = pytest.mark.gpu


def fill(dev, *shape):
    import torch
    t = torch.empty(shape, dtype=torch.bfloat16, device=dev)
    for row in t.view(-1, shape[-1]):
        row.normal_()
    return t


def test_recurrence_past_32_bit_offsets(dev):
    """Five rows of 2^29 tokens: the last row's outputs and gradients have the bits of that row alone, cut alike."""
    import torch
    import selective_state_space_75_amd as m
    D, L = 5, 1 << 29
    torch.manual_seed(0)
    x, r, dy = (fill(dev, 1, D, L) for _ in range(3))
    A = -torch.rand(D, device=dev) - 0.1
    last = lambda t: t[:, D - 1:].contiguous()  # noqa: E731
    with m.glr_test_knobs(waves=16, segments=128):
        y, h = m.glr_fwd(x, r, None, A, return_final_state=True)
        y1, h1 = m.glr_fwd(last(x), last(r), None, A[D - 1:].contiguous(), return_final_state=True)
        assert torch.equal(y[:, D - 1:], y1) and torch.equal(h[:, D - 1:], h1)
    del y
    with m.glr_test_knobs(waves=16):
        g = m.glr_bwd(x, r, None, A, None, None, None, dy)
        g1 = m.glr_bwd(last(x), last(r), None, A[D - 1:].contiguous(), None, None, None, last(dy))
        assert torch.equal(g["dx"][:, D - 1:], g1["dx"]) and torch.equal(g["dr"][:, D - 1:], g1["dr"])
    del g, g1
    # a window at the end against the oracle: what is 4000 tokens back is forgotten (decays below e^-0.05 on average)
    w = slice(L - 6000, L)
    yr, hr = O.glr(from_dev(x[:, :, w]), from_dev(r[:, :, w]), None, from_dev(A))
    near(y1[:, :, L - 1000:].float(), yr[:, D - 1:, -1000:], 2.0 ** -8 + E, "window")
    near(h, hr, E, "final state")


def test_short_rows_past_32_bit_offsets(dev):
    """The last rows have the bits that they have alone."""
    import torch
    import selective_state_space_75_amd as m
    D, L = 23000000, 99
    torch.manual_seed(3)
    x, r, dy = (torch.randn(1, 1000, L, device=dev).bfloat16().repeat(1, D // 1000, 1) for _ in range(3))
    A = -torch.rand(D, device=dev) - 0.1
    cut = lambda t: t[:, D - 300:].contiguous()  # noqa: E731
    y, h = m.glr_fwd(x, r, x, A, return_final_state=True)
    y1, h1 = m.glr_fwd(cut(x), cut(r), cut(x), A[D - 300:].contiguous(), return_final_state=True)
    assert torch.equal(cut(y), y1) and torch.equal(h[:, D - 300:], h1)
    del y
    g = m.glr_bwd(x, r, None, A, None, None, None, dy)
    g1 = m.glr_bwd(cut(x), cut(r), None, A[D - 300:].contiguous(), None, None, None, cut(dy))
    for n in ("dx", "dr"):
        assert torch.equal(cut(g[n]), g1[n]), n
    assert torch.equal(g["dA"][D - 300:], g1["dA"])


def test_norm_past_32_bit_offsets(dev):
    import torch
    import selective_state_space_75_amd as m
    D, L = 9, 1 << 28                      # 2^29 tokens would be a launch of 2^32 threads
    torch.manual_seed(1)
    x, dy = fill(dev, 1, D, L), fill(dev, 1, D, L)
    w = torch.randn(D, device=dev)
    for part in (slice(L - 700, L), slice(L // 2 - 300, L // 2 + 300)):
        xs, ds = from_dev(x[:, :, part]), from_dev(dy[:, :, part])
        y = m.layer_norm_fwd(x, w)
        near(y[:, :, part].float(), O.layer_norm(xs, from_dev(w)), 2.0 ** -8 + E, "y")
        del y
        g = m.layer_norm_bwd(x, w, None, None, dy)
        ref = O.layer_norm_bwd(xs, from_dev(w), None, None, ds)
        near(g["dx"][:, :, part].float(), ref["dx"], 2.0 ** -8 + E, "dx", ref["scale"]["dx"])
        del g


def test_update_in_a_pool_past_32_bit_offsets(dev):
    import torch
    import selective_state_space_75_amd as m
    S, D, B = 530_000, 4096, 3
    pool = torch.empty((S, D), device=dev)
    slots = torch.tensor([S - 1, 0, S - 2], dtype=torch.int32, device=dev)
    rng = np.random.default_rng(0)
    h0 = rng.standard_normal((B, D)).astype(np.float32)
    pool[slots.long()] = torch.from_numpy(h0).to(dev)
    x, r = (torch.from_numpy(rng.standard_normal((B, D)).astype(np.float32)).to(dev) for _ in range(2))
    A = -torch.rand(D, device=dev) - 0.1
    y = m.glr_update(pool, x, r, None, A, slots=slots)
    yr, hr = O.glr(from_dev(x)[..., None], from_dev(r)[..., None], None, from_dev(A), initial_state=h0)
    near(y, yr[..., 0], E, "y")
    near(pool[slots.long()], hr, E, "state")


@pytest.mark.parametrize("rows,D,gated", [(1800000, 1300, False), (260000, 9000, True)])
def test_token_major_norm_past_32_bit_offsets(rows, D, gated, dev):
    """The last tokens have the bits that they have alone."""
    import torch
    import selective_state_space_75_amd as m
    torch.manual_seed(2)
    x, dy = (torch.randn(3000, D, device=dev).bfloat16().repeat((rows + 2999) // 3000, 1)[:rows] for _ in range(2))
    w = torch.randn(D, device=dev)
    z = dy if gated else None
    cut = lambda t: None if t is None else t[rows - 3:].contiguous()  # noqa: E731
    y = m.layer_norm_fwd(x, w, w, z)
    assert torch.equal(y[rows - 3:], m.layer_norm_fwd(cut(x), w, w, cut(z)))
    del y
    g = m.layer_norm_bwd(x, w, w, z, dy)
    g1 = m.layer_norm_bwd(cut(x), w, w, cut(z), cut(dy))
    for n in ("dx", "dz"):
        assert g[n] is None or torch.equal(g[n][rows - 3:], g1[n]), n
