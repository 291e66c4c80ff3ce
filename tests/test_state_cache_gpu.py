"""The 8-bit state cache on the GPU: codes and exponents equal the oracle's bit for
bit (a division by a power of two is exact, so there is one right code), and
reading is exact."""
import numpy as np
import pytest

from helpers import from_dev, log, to_dev
from oracle import gdr as O

pytestmark = pytest.mark.gpu


def _state(rows, n, seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, n)) * np.exp2(rng.integers(-20, 20, (rows, (n + 31) // 32)).repeat(32, 1)[:, :n])
    return x.astype(np.float32)


@pytest.mark.parametrize("rows,n,dtype", [(1, 1, "f32"), (3, 31, "f32"), (2, 32, "bf16"), (4, 133, "f32"),
                                          (2, 1000, "bf16"), (3, 4096, "f32"), (2, 5004, "f32"), (1, 70002, "f32"),
                                          (70, 131072, "f32")])
def test_write_and_read(rows, n, dtype, dev):
    import torch
    import selective_state_space_75_amd as m
    log("[cache] rows=%d n=%d %s" % (rows, n, dtype))
    S = rows + 3
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    x = to_dev(_state(rows, n, n), dev).to(dt)
    slots = np.random.default_rng(n).permutation(S)[:rows].astype(np.int32)
    if rows > 1:
        slots[1] = -1
    if rows > 2:
        slots[2] = S
    codes = torch.full((S, n), 99, dtype=torch.int8, device=dev)
    exps = torch.full((S, (n + 31) // 32), 77, dtype=torch.uint8, device=dev)
    sl = torch.from_numpy(slots).to(dev)
    m.state_cache_write(x, codes, exps, slots=sl)
    back = m.state_cache_read(codes, exps, slots=sl, dtype=dt)
    torch.cuda.synchronize()
    c, e, xr, b = codes.cpu().numpy(), exps.cpu().numpy(), from_dev(x), from_dev(back)
    used = []
    for r in range(rows):
        if not 0 <= slots[r] < S:
            assert not b[r].any()
            continue
        used.append(slots[r])
        if n <= 6000 or r == 0:
            cr, er = O.cache_write(xr[r])
            assert np.array_equal(c[slots[r]], cr) and np.array_equal(e[slots[r]], er)
        assert np.array_equal(b[r], O.cache_read(c[slots[r]], e[slots[r]]))
        step = np.exp2(e[slots[r]].astype(np.float64) - 127).repeat(32)[:n]
        assert np.all(np.abs(b[r] - xr[r]) <= step / 2)
    idle = sorted(set(range(S)) - set(used))
    assert (c[idle] == 99).all() and (e[idle] == 77).all()


def test_extremes(dev):
    """Zeros, the smallest and largest numbers, ties, a group whose maximum is at 127 steps or
    just above, infinities and NaN (the group reads back as NaN, its neighbours do not)."""
    import torch
    import selective_state_space_75_amd as m
    x = np.zeros((1, 32 * 8 + 5), dtype=np.float32)
    x[0, 32:36] = [127.0, 0.5, 1.5, -2.5]
    x[0, 64:66] = [np.nextafter(np.float32(127), np.float32(200)), 1.0]
    x[0, 96:98] = [np.finfo(np.float32).max, -1.0]
    x[0, 128:130] = [1e-45, -1e-38]
    x[0, 160:162] = [np.inf, 3.0]
    x[0, 192:194] = [np.nan, 3.0]
    x[0, 224] = -3.0
    x[0, 256:] = [1, 2, 3, 4, 5]
    codes, exps = m.state_cache(1, x.shape[1], dev)
    assert not m.state_cache_read(codes, exps).any()           # an empty cache reads as zeros
    m.state_cache_write(to_dev(x, dev), codes, exps)
    back = from_dev(m.state_cache_read(codes, exps))[0]
    cr, er = O.cache_write(x[0])
    assert np.array_equal(codes.cpu().numpy()[0], cr) and np.array_equal(exps.cpu().numpy()[0], er)
    assert np.isnan(back[160:224]).all() and np.isfinite(back[:160]).all() and np.isfinite(back[224:]).all()
    assert np.array_equal(back[32:36], [127, 0, 2, -2])
    assert torch.equal(m.state_cache_read(codes, exps, dtype=torch.bfloat16).float().nan_to_num(7.0),
                       m.state_cache_read(codes, exps).nan_to_num(7.0))


def test_shared_slots_and_states_of_every_layer(dev):
    """Rows that share a slot read the same numbers; states of any trailing shape are taken flat."""
    import torch
    import selective_state_space_75_amd as m
    st = to_dev(_state(3, 8 * 16, 5), dev).view(3, 8, 16)
    codes, exps = m.state_cache(4, 8 * 16, dev)
    m.state_cache_write(st, codes, exps)
    sl = torch.tensor([2, 0, 2, -1, 2], dtype=torch.int32, device=dev)
    out = torch.full((5, 8, 16), 7.0, device=dev)
    assert m.state_cache_read(codes, exps, slots=sl, out=out) is out
    torch.cuda.synchronize()
    assert torch.equal(out[0], out[2]) and torch.equal(out[0], out[4]) and not out[3].any()
    assert float((out[1] - st[0]).abs().max() / st[0].abs().max()) <= 1 / 127


def test_refusals(dev):
    import torch
    import selective_state_space_75_amd as m
    codes, exps = m.state_cache(2, 64, dev)
    with pytest.raises(ValueError):
        m.state_cache_write(torch.zeros(2, 63, device=dev), codes, exps)
    with pytest.raises(TypeError):
        m.state_cache_write(torch.zeros(2, 64, device=dev, dtype=torch.float16), codes, exps)
    with pytest.raises(m.MambaError):
        m.state_cache_write(torch.zeros(3, 64, device=dev), codes, exps)       # no third slot
    with pytest.raises(TypeError):
        m.state_cache_read(codes, exps, slots=torch.zeros(2, dtype=torch.int64, device=dev))
