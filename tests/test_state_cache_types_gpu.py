"""The state cache's kernels by type and form: element by element (n off 4, or a misaligned state) and
vectors, one or four pieces per thread, in fp32 and bf16; codes and what is read back are exact."""
import numpy as np
import pytest

from helpers import from_dev, log
from oracle import gdr as O

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,n,shift", [
    (4, 133, 0),                  # element by element
    (3, 1000, 1),                 # the same: the state one element off its alignment
    (2, 1000, 0),                 # vectors, one piece per thread
    (70, 131072, 0),              # vectors, four pieces
    (130, 65540, 0),              # the same, the last workgroup of a row nearly empty
    (70, 131073, 0),              # as many numbers, element by element
])
def test_forms(rows, n, shift, dtype, dev):
    import torch
    import selective_state_space_75_amd as m
    log("[cache forms] rows=%d n=%d shift=%d %s" % (rows, n, shift, dtype))
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    gen = torch.Generator(device=dev).manual_seed(n + rows)
    flat = torch.randn(rows * n + shift, generator=gen, device=dev)
    flat = (flat * torch.exp2(torch.randint(-20, 20, flat.shape, generator=gen, device=dev).float())).to(dt)
    x = flat[shift:].view(rows, n)
    S = rows + 2
    slots = torch.randperm(S, generator=gen, device=dev)[:rows].int()
    codes = torch.full((S, n), 99, dtype=torch.int8, device=dev)
    exps = torch.full((S, (n + 31) // 32), 77, dtype=torch.uint8, device=dev)
    m.state_cache_write(x, codes, exps, slots=slots)
    out = torch.empty(rows * n + shift, dtype=dt, device=dev)[shift:].view(rows, n)
    m.state_cache_read(codes, exps, slots=slots, out=out)
    torch.cuda.synchronize()
    where = slots.long()
    for r in (0, rows - 1):
        s = int(where[r])
        cr, er = O.cache_write(from_dev(x[r, -8192 - n % 32:]) if n > 8192 else from_dev(x[r]))
        # (the last 8192 numbers and a few more, from a group's start)
        assert np.array_equal(codes[s].cpu().numpy()[-cr.size:], cr) and np.array_equal(exps[s].cpu().numpy()[-er.size:], er)
    # all rows: a code times its power of two, and within half a step
    step = torch.exp2(exps[where].double() - 127).repeat_interleave(32, 1)[:, :n]
    assert torch.equal(codes[where].double() * step, out.double())
    assert ((out.double() - x.double()).abs() <= step / 2).all()
    idle = sorted(set(range(S)) - set(slots.tolist()))
    assert (codes[idle] == 99).all() and (exps[idle] == 77).all()
