"""The gated linear recurrence and the layer norm as they are used together: a prompt through norm,
projection, convolution, recurrence and the norm per head, its state parked in 8 bits and taken back,
tokens one by one; training forward and backward; all of it captured into a graph; and on streams of its own.

Bars are those of the single calls, because every step is compared with the fp64 oracle from the GPU's
own inputs of that step; graph replays and other streams give the same bits."""
import numpy as np
import pytest

from helpers import F32_REL_L2, assert_close, f64, from_dev, log, rel_l2, to_dev
from oracle import gdr as C
from oracle import glr as O
from selective_state_space_75_amd import workloads as W

pytestmark = pytest.mark.gpu


def n64(t):
    return f64(from_dev(t))


@pytest.mark.parametrize("B,D,L,heads,K", [(3, 96, 75, 4, 4), (2, 640, 12, 5, 3)])
def test_prompt_park_and_decode(B, D, L, heads, K, dev):
    import torch
    import selective_state_space_75_amd as m
    T, S = 3, B + 2
    rng = np.random.default_rng(B * L)
    f32 = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(dev)  # noqa: E731
    x, w_in = f32(B, D, L + T).bfloat16(), f32(4 * D, D) * D ** -0.5
    wn, bn, wh, wc = 1 + 0.1 * f32(D), 0.1 * f32(D), 1 + 0.1 * f32(D), 0.5 * f32(D, K)
    A, rb, ib = -f32(D).abs() - 0.01, f32(D), f32(D)

    def project(n):                       # channel-major: (4 D, D) x (B, D, L)
        return torch.stack([torch.mm(w_in, row.float()) for row in n]).bfloat16()

    n = m.layer_norm_fwd(x[:, :, :L].contiguous(), wn, bn)
    assert_close(from_dev(n), O.layer_norm(n64(x[:, :, :L]), n64(wn), n64(bn)), True, "norm")
    p = project(n)
    u, cs = m.conv1d_fwd(p[:, :D].contiguous(), wc, return_final_state=True)
    y, h = m.glr_fwd(u, p[:, D:2 * D], p[:, 2 * D:3 * D], A, rb, ib, return_final_state=True)
    yr, hr = O.glr(n64(u), n64(p[:, D:2 * D]), n64(p[:, 2 * D:3 * D]), n64(A), n64(rb), n64(ib))
    assert_close(from_dev(y), yr, True, "recurrence")
    assert rel_l2(from_dev(h), hr) <= F32_REL_L2
    o = m.layer_norm_fwd(y, wh, None, p[:, 3 * D:], groups=heads, rms=True)
    assert_close(from_dev(o), O.layer_norm(n64(y), n64(wh), None, n64(p[:, 3 * D:]), groups=heads, rms=True), True, "heads")

    slots = torch.from_numpy(rng.permutation(S)[:B].astype(np.int32)).to(dev)
    codes, exps = m.state_cache(S, D, dev)
    m.state_cache_write(h, codes, exps, slots=slots)
    pool = torch.full((S, D), 7.0, device=dev)
    pool[slots.long()] = m.state_cache_read(codes, exps, slots=slots)
    for b in range(B):
        assert np.array_equal(from_dev(pool)[int(slots[b])], C.cache_read(*C.cache_write(from_dev(h)[b])))
    for t in range(L, L + T):
        n = m.layer_norm_fwd(x[:, :, t].contiguous(), wn, bn)             # one token a row: (B, D)
        assert_close(from_dev(n), O.layer_norm(n64(x[:, :, t]), n64(wn), n64(bn)), True, "norm, token %d" % t)
        p = torch.mm(n.float(), w_in.t().contiguous()).bfloat16()
        u = m.conv1d_update(cs, p[:, :D].contiguous(), wc)
        before = n64(pool)[slots.cpu().numpy()]
        y = m.glr_update(pool, u, p[:, D:2 * D], p[:, 2 * D:3 * D], A, rb, ib, slots=slots)
        args = [n64(v)[..., None] for v in (u, p[:, D:2 * D], p[:, 2 * D:3 * D])]
        yr, hr = O.glr(*args, n64(A), n64(rb), n64(ib), initial_state=before)
        assert_close(from_dev(y), yr[..., 0], True, "recurrence, token %d" % t)
        assert rel_l2(n64(pool)[slots.cpu().numpy()], hr) <= F32_REL_L2
        o = m.layer_norm_fwd(y, wh, None, p[:, 3 * D:], groups=heads, rms=True)
        assert_close(from_dev(o), O.layer_norm(n64(y), n64(wh), None, n64(p[:, 3 * D:]), groups=heads, rms=True), True,
                     "heads, token %d" % t)
    rest = np.setdiff1d(np.arange(S), slots.cpu().numpy())
    assert (from_dev(pool)[rest] == 7.0).all()


def test_training_step(dev):
    """fp32 gradients through norm, recurrence and the gated norm per head against the oracle's chain from the
    start: each of the three stages adds about its own bar, 1e-5 of the size of the terms it sums."""
    import torch
    import selective_state_space_75_amd as m
    B, D, L, heads = 2, 48, 150, 4
    v = W.glr_inputs(B, D, L, "f32", 70)
    x = W.norm_inputs((B, D, L), "f32", 71)
    t, q = {k: to_dev(a, dev) for k, a in v.items()}, {k: to_dev(a, dev) for k, a in x.items()}
    n = m.layer_norm_fwd(q["x"], q["weight"], q["bias"])
    gates = (t["r"], t["i"], t["A"], t["r_bias"], t["i_bias"])
    y = m.glr_fwd(n, *gates)
    g2 = m.layer_norm_bwd(y, q["weight"], None, t["z"], t["dy"], groups=heads, rms=True)
    g1 = m.glr_bwd(n, *gates, None, g2["dx"])
    g0 = m.layer_norm_bwd(q["x"], q["weight"], q["bias"], None, g1["dx"])
    nr = O.layer_norm(f64(x["x"]), f64(x["weight"]), f64(x["bias"]))
    og = [f64(v[k]) for k in ("r", "i", "A", "r_bias", "i_bias")]
    yr, _ = O.glr(nr, *og)
    r2 = O.layer_norm_bwd(yr, f64(x["weight"]), None, f64(v["z"]), f64(v["dy"]), groups=heads, rms=True)
    r1 = O.glr_bwd(nr, *og, None, r2["dx"])
    r0 = O.layer_norm_bwd(f64(x["x"]), f64(x["weight"]), f64(x["bias"]), None, r1["dx"])
    for name, got, ref in ([("heads " + k, g2[k], r2) for k in ("dz", "dweight", "dbias")]
                           + [("recurrence " + k, g1[k], r1) for k in ("dr", "di", "dA", "dr_bias", "di_bias")]
                           + [("norm " + k, g0[k], r0) for k in ("dx", "dweight", "dbias")]):
        k = name.split()[1]
        size = np.linalg.norm(ref["scale"].get(k, ref[k]))
        err = np.linalg.norm(from_dev(got) - ref[k])
        log("  %s: off by %.2e of its terms" % (name, err / size))
        assert err <= 3 * F32_REL_L2 * size, name


def all_calls(m, t, q, rows, one, state, slots, ws, heads=3, **kw):
    """Every call of both operators, each layout of the norm."""
    gates = (t["r"], t["i"], t["A"], t["r_bias"], t["i_bias"], t["z"])
    out = list(m.glr_fwd(t["x"], *gates, initial_state=t["initial_state"], return_final_state=True,
                         workspace=ws[0], **kw))
    g = m.glr_bwd(t["x"], *gates, t["dy"], initial_state=t["initial_state"], dfinal_state=t["dfinal_state"],
                  workspace=ws[1], **kw)
    out += [g[k] for k in sorted(g)]
    out.append(m.glr_update(state, one["x"], one["r"], one["i"], *gates[2:5], one["z"], slots=slots, **kw))
    for x, groups in ((q, 1), (q, heads), (rows, 1)):
        out.append(m.layer_norm_fwd(x["x"], x["weight"], x["bias"], x["z"], groups=groups, **kw))
        g = m.layer_norm_bwd(x["x"], x["weight"], x["bias"], x["z"], x["dy"], groups=groups, **kw)
        out += [g[k] for k in sorted(g)]
    return out


def make(B, D, L, seed, dev):
    t = {k: to_dev(a, dev) for k, a in W.glr_inputs(B, D, L, "bf16", seed).items()}
    q = {k: to_dev(a, dev) for k, a in W.norm_inputs((B, D, L), "bf16", seed + 1).items()}
    rows = {k: to_dev(a, dev) for k, a in W.norm_inputs((B * 20, D), "bf16", seed + 2).items()}
    one = {k: t[k][:, :, 0].contiguous() for k in ("x", "r", "i", "z")}
    return t, q, rows, one


@pytest.mark.parametrize("D,waves,segments", [(45, 0, 0), (45, 1, 3), (2100, 0, 0)])
def test_graph_replays_equal_eager(D, waves, segments, dev):
    import torch
    import selective_state_space_75_amd as m
    B, L = 2, 700
    sets = [make(B, D, L, 40 + 5 * k, dev) for k in range(3)]
    bufs = [{n: a.clone() for n, a in d.items()} for d in sets[0]]
    pool = torch.randn(4, D, device=dev)
    slots = torch.tensor([3, 1], dtype=torch.int32, device=dev)
    state = pool.clone()
    with m.glr_test_knobs(waves=waves, segments=segments):
        need = [m.glr_workspace_size(B, D, L), m.glr_bwd_workspace_size(B, D, L)]
        ws = [torch.empty(max(n, 1), dtype=torch.uint8, device=dev) for n in need]
        side = torch.cuda.Stream(dev)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs = all_calls(m, *bufs, state, slots, ws)
        for rep in range(5):
            src = sets[rep % 3]
            for b, s in zip(bufs, src):
                for n in b:
                    b[n].copy_(s[n])
            state.copy_(pool)
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            got = [o.clone() for o in outs] + [state.clone()]
            st2 = pool.clone()
            ref = all_calls(m, *src, st2, slots, [None, None]) + [st2]
            torch.cuda.synchronize()
            assert len(got) == len(ref)
            for i, (a, r) in enumerate(zip(got, ref)):
                assert torch.equal(a, r), "replay %d, output %d" % (rep, i)


@pytest.mark.parametrize("D", [90, 1500])
def test_two_streams_at_once(D, dev):
    """Calls on two streams at once, the wrappers' own workspaces: the bits of one call alone."""
    import torch
    import selective_state_space_75_amd as m
    B, L = 3, 1300
    sets = [make(B, D, L, 60 + 5 * k, dev) for k in range(2)]
    pool = torch.randn(B, D, device=dev)

    def run(s, stream):
        state = pool.clone()
        if stream is not None:                           # the state is made on the caller's stream
            stream.wait_stream(torch.cuda.current_stream(dev))
        return all_calls(m, *s, state, None, [None, None], stream=stream) + [state]

    alone = [run(s, None) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(dev) for _ in sets]
    for _ in range(3):
        got = [run(s, st) for s, st in zip(sets, streams)]
        # the caller's stream allocates meanwhile: none of it may be a running call's workspace
        junk = [torch.full((1 << 20,), float("nan"), device=dev) for _ in range(8)]
        torch.cuda.synchronize()
        del junk
        for a, b in zip(alone, got):
            assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_workspaces_are_checked(dev):
    import torch
    import selective_state_space_75_amd as m
    x = torch.zeros(1, 2, 1 << 15, device=dev)
    A = -torch.ones(2, device=dev)
    need = m.glr_workspace_size(1, 2, 1 << 15)
    assert need > 0
    with pytest.raises(m.MambaError):
        m.glr_fwd(x, x, None, A, workspace=torch.empty(need - 1, dtype=torch.uint8, device=dev))
    with pytest.raises(ValueError, match="workspace is on"):
        m.glr_fwd(x, x, None, A, workspace=torch.empty(need, dtype=torch.uint8))
    big = torch.zeros(1, 10000, 16, device=dev)
    need = m.layer_norm_workspace_size(1, 10000, 16)
    assert need > 0
    with pytest.raises(m.MambaError):
        m.layer_norm_fwd(big, workspace=torch.empty(need - 1, dtype=torch.uint8, device=dev))
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        m.layer_norm_fwd(big, workspace=torch.empty(2 * need, dtype=torch.uint8, device=dev)[::2])
