"""The selective state-space scan on the GPU (gla_ssm_fwd, gla_ssm_varlen,
gla_ssm_step) against its definition in float64, and the properties that tie
the three together."""
import pytest
import torch

import ssm_plain as plain
from ssm_plain import close, d

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def gla():
    import linear_attention_chunk_gb300 as m
    from linear_attention_chunk_gb300.build import build
    build()
    return m


def inputs(lead, D, N, dtype, seed, gate=True, bias=True, skip=True):
    g = torch.Generator().manual_seed(seed)

    def rn(*shape, std=1.0, dt=dtype):
        return (torch.randn(*shape, generator=g) * std).to(dt).cuda()
    step = torch.exp(torch.rand(D, generator=g) * 4.6 - 6.9)
    return dict(x=rn(*lead, D), dt=rn(*lead, D, std=0.7), Bm=rn(*lead, N), Cm=rn(*lead, N),
                A=(-torch.arange(1, N + 1).float() * torch.exp(torch.randn(D, N, generator=g) * 0.1)).cuda(),
                skip=(1 + rn(D, std=0.1, dt=FP)) if skip else None, z=rn(*lead, D) if gate else None,
                dt_bias=(step + torch.log(-torch.expm1(-step))).cuda() if bias else None)


def ref_fwd(s, h0, soft=True):
    B = s["x"].shape[0]
    D, N = s["A"].shape
    out = []
    for b in range(B):
        h = torch.zeros(D, N, dtype=plain.F64) if h0 is None else d(h0[b])
        out.append(plain.scan(d(s["x"][b]), d(s["dt"][b]), d(s["A"]), d(s["Bm"][b]), d(s["Cm"][b]), d(s["skip"]),
                              None if s["z"] is None else d(s["z"][b]), d(s["dt_bias"]), h, soft))
    return [torch.stack(v) for v in zip(*out)]


def call_fwd(gla, s, h0=None, **kw):
    return gla.gla_ssm_fwd(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["skip"], s["z"], s["dt_bias"], h0, **kw)


@pytest.mark.parametrize("dtype,B,T,D,N,gate,bias,skip,state", [
    (BF, 1, 1, 8, 16, True, True, True, False), (FP, 2, 33, 72, 16, True, True, True, True),
    (BF, 3, 31, 64, 8, False, True, True, True), (FP, 1, 64, 200, 32, True, False, False, False),
    (BF, 2, 129, 136, 16, True, True, False, True), (FP, 1, 7, 1032, 8, False, False, True, True),
    (BF, 1, 700, 24, 16, True, True, True, True), (FP, 2, 1025, 40, 16, True, True, True, False),
    (BF, 1, 300, 16, 32, True, True, True, True), (FP, 2, 70, 4, 8, True, True, True, True),
    (FP, 1, 45, 516, 16, True, True, True, True)])
def test_fwd_matches_the_definition(gla, dtype, B, T, D, N, gate, bias, skip, state):
    s = inputs((B, T), D, N, dtype, 100 + T, gate, bias, skip)
    h0 = torch.randn(B, D, N, generator=torch.Generator().manual_seed(T)).cuda() if state else None
    y, hT = call_fwd(gla, s, h0)
    gla.gla_check()
    ry, my, rh, mh = ref_fwd(s, h0)
    close(y, ry, my, T, "y")
    close(hT, rh, mh, T, "hT")


@pytest.mark.parametrize("B,T,D", [(1, 2500, 64), (2, 1111, 136)])
def test_segments_agree_with_one_chain_and_update_the_state_in_place(gla, B, T, D):
    s = inputs((B, T), D, 16, FP, 7)
    h0 = torch.randn(B, D, 16, generator=torch.Generator().manual_seed(3)).cuda()
    assert gla.gla_ssm_fwd_workspace_size(B, T, D, 16, gla.GLA_FP32) > 0
    y, hT = call_fwd(gla, s, h0)
    assert gla.gla_last_launch_count() == 2
    none = torch.empty(0, dtype=torch.uint8, device="cuda")
    y1, hT1 = call_fwd(gla, s, h0, workspace=none)
    assert gla.gla_last_launch_count() == 1
    state = h0.clone()
    y2, _ = call_fwd(gla, s, state, hT=state)
    gla.gla_check()
    ry, my, rh, mh = ref_fwd(s, h0)
    for got, h in ((y, hT), (y1, hT1), (y2, state)):
        close(got, ry, my, T, "y")
        close(h, rh, mh, T, "hT")
    assert torch.equal(y, y2) and torch.equal(hT, state)


def test_strided_rows_give_the_same_bits(gla):
    B, T, D, N = 2, 50, 72, 16
    s = inputs((B, T), D, N, BF, 11)
    y, hT = call_fwd(gla, s)
    xz = torch.randn(B, T, 2 * D + 16, device="cuda").to(BF)
    dbc = torch.randn(B, T, 5 + 2 * N, device="cuda").to(BF)
    xz[..., :D], xz[..., D + 16:] = s["x"], s["z"]
    dbc[..., 5:5 + N], dbc[..., 5 + N:] = s["Bm"], s["Cm"]
    t = dict(s, x=xz[..., :D], z=xz[..., D + 16:], Bm=dbc[..., 5:5 + N], Cm=dbc[..., 5 + N:])
    y1, h1 = call_fwd(gla, t)
    gla.gla_check()
    assert torch.equal(y, y1) and torch.equal(hT, h1)
    with pytest.raises(gla.GlaError):                       # sequences not a whole number of rows apart
        call_fwd(gla, dict(s, x=xz[:, ::2, :D][:, :T // 2]))
    with pytest.raises(gla.GlaError):                       # channels not adjacent
        call_fwd(gla, dict(s, x=torch.randn(B, T, 2 * D, device="cuda").to(BF)[..., ::2]))


def test_empty_calls(gla):
    s = inputs((2, 5), 16, 16, BF, 1)
    h0 = torch.randn(2, 16, 16, device="cuda")
    e = {k: (v[:, :0] if k in ("x", "dt", "z", "Bm", "Cm") else v) for k, v in s.items()}
    y, hT = call_fwd(gla, e, h0)
    gla.gla_check()
    assert y.shape == (2, 0, 16) and torch.equal(hT, h0)
    assert not call_fwd(gla, e)[1].any()
    e = {k: (v[:0] if k in ("x", "dt", "z", "Bm", "Cm") else v) for k, v in s.items()}
    assert call_fwd(gla, e)[0].shape == (0, 5, 16)


def test_extreme_steps_and_raw_steps(gla):
    """A step of zero keeps the state, a long one clears it; without softplus dt is the step itself."""
    T, D, N = 40, 16, 16
    s = inputs((1, T), D, N, FP, 5, bias=False)
    s["dt"][0, 10:20] = -300.0                              # softplus underflows to 0
    s["dt"][0, 25] = 90.0                                   # decay e^-90 and less
    h0 = torch.randn(1, D, N, device="cuda")
    y, hT = call_fwd(gla, s, h0)
    ry, my, rh, mh = ref_fwd(s, h0)
    close(y, ry, my, T, "y")
    close(hT, rh, mh, T, "hT")
    s["dt"] = torch.rand(1, T, D, device="cuda") * 0.2
    s["dt"][0, 3] = 0.0
    y, hT = call_fwd(gla, s, h0, softplus=False)
    gla.gla_check()
    ry, my, rh, mh = ref_fwd(s, h0, soft=False)
    close(y, ry, my, T, "y")
    close(hT, rh, mh, T, "hT")


def test_a_nan_stays_in_its_channel_and_sequence(gla):
    s = inputs((2, 70), 64, 16, FP, 9)
    y, hT = call_fwd(gla, s)
    s["x"][1, 30, 5] = float("nan")
    y1, h1 = call_fwd(gla, s)
    gla.gla_check()
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[1, 30:, 5] = True
    assert torch.equal(torch.isnan(y1), bad)
    assert torch.equal(y1[~bad], y[~bad]) and torch.isnan(h1[1, 5]).all() and torch.isnan(h1).sum() == 16


# ----------------------------------------------------------- packed prompts
def pools(n, D, N, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(n, D, N, generator=g).cuda(), torch.randn(n, 4, D, generator=g).cuda(),
            (torch.randn(D, 4, generator=g) * 0.5).cuda(), (torch.randn(D, generator=g) * 0.1).cuda())


def ref_packed(s, cu, slots, pool, win, w, b):
    """Per sequence: y, magnitudes, state, its magnitudes, window."""
    out = []
    for i, sl in enumerate(slots):
        r = slice(cu[i], cu[i + 1])
        x = d(s["x"][r])
        u, um, nw = (x, None, None) if w is None else plain.conv(x, d(w), d(b), d(win[sl]))
        out.append(plain.scan(u, d(s["dt"][r]), d(s["A"]), d(s["Bm"][r]), d(s["Cm"][r]), d(s["skip"]),
                              None if s["z"] is None else d(s["z"][r]), d(s["dt_bias"]), d(pool[sl]), True, um) + (nw,))
    return out


def call_varlen(gla, s, cu, pool, slots=None, w=None, b=None, win=None, **kw):
    return gla.gla_ssm_varlen(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], cu, pool, s["skip"], s["z"], s["dt_bias"],
                              slots, conv_w=w, conv_b=b, win_pool=win, **kw)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype,lens,D,N,filt", [
    (BF, [5, 0, 1, 64, 3, 0], 72, 16, True), (FP, [1], 8, 8, True), (FP, [2, 1, 3, 1], 64, 16, True),
    (BF, [1300, 2, 513, 0, 40], 40, 16, True), (FP, [700, 1, 600], 24, 32, True), (BF, [33, 200, 7], 136, 16, False),
    (FP, [0, 0, 9], 16, 16, False), (FP, [2, 90, 1], 68, 8, True)])
def test_varlen_matches_the_definition(gla, dtype, lens, D, N, filt):
    cu = [0]
    for v in lens:
        cu.append(cu[-1] + v)
    extra = 3                                               # rows behind the last sequence
    s = inputs((cu[-1] + extra,), D, N, dtype, 40 + len(lens))
    n = len(lens)
    slots = [(3 * i + 1) % (n + 2) if (n + 2) % 3 else n + 1 - i for i in range(n)]
    assert len(set(slots)) == n
    pool, win, w, b = pools(n + 2, D, N, 8)
    if not filt:
        w = b = win = None
    p1, w1 = pool.clone(), None if win is None else win.clone()
    y = torch.full((cu[-1] + extra, D), 7.0, dtype=dtype, device="cuda")
    call_varlen(gla, s, i32(cu), p1, i32(slots), w, b, w1, y=y)
    gla.gla_check()
    for i, (ry, my, rh, mh, nw) in enumerate(ref_packed(s, cu, slots, pool, win, w, b)):
        close(y[cu[i]:cu[i + 1]], ry, my, lens[i], f"y of {i}")
        if lens[i]:
            close(p1[slots[i]], rh, mh, lens[i], f"state of {i}")
            if filt:
                assert torch.equal(d(w1[slots[i]]), nw)     # inputs, unrounded
        else:
            assert torch.equal(p1[slots[i]], pool[slots[i]])
            assert w1 is None or torch.equal(w1[slots[i]], win[slots[i]])
    assert (y[cu[-1]:] == 7).all()
    rest = [k for k in range(n + 2) if k not in slots]
    assert torch.equal(p1[rest], pool[rest]) and (w1 is None or torch.equal(w1[rest], win[rest]))


def test_bad_entries_skip_their_sequence_and_are_reported(gla):
    D, N = 24, 16
    s = inputs((30,), D, N, FP, 3)
    pool, win, w, b = pools(3, D, N, 2)
    good = [(pool.clone(), win.clone()) for _ in range(1)][0]
    y0 = call_varlen(gla, s, i32([0, 10, 20, 30]), good[0], i32([0, 1, 2]), w, b, good[1])
    gla.gla_check()
    for cu, slots, hurt in (([0, 10, 20, 99], [0, 1, 2], 2), ([0, 10, 20, 30], [0, 3, 2], 1),
                            ([0, 10, 20, 30], [-1, 1, 2], 0)):
        p1, w1 = pool.clone(), win.clone()
        y = torch.zeros(30, D, device="cuda")
        call_varlen(gla, s, i32(cu), p1, i32(slots), w, b, w1, y=y)
        with pytest.raises(gla.GlaError) as e:
            gla.gla_check()
        assert e.value.status == gla.GLA_ERR_INVALID_ARG
        for i in range(3):
            r = slice(10 * i, 10 * i + 10)
            if i == hurt:
                assert not y[r].any() and torch.equal(p1[i], pool[i]) and torch.equal(w1[i], win[i])
            else:
                assert torch.equal(y[r], y0[r]) and torch.equal(p1[i], good[0][i]) and torch.equal(w1[i], good[1][i])
    with pytest.raises(gla.GlaError):                       # a decreasing offset
        call_varlen(gla, s, i32([0, 20, 10, 30]), pool.clone(), None, w, b, win.clone())
        gla.gla_check()
    gla.gla_check()                                         # reported once


@pytest.mark.parametrize("cu", [[0, 1000, 0, 1000], [0, 20, 10, 1000], [500, 1000, 400, 300]])
def test_decreasing_offsets_run_no_sequence(gla, cu):
    """Overlapping sequences of several segments would mix in the workspace and in y: pools, windows and y
    are left alone, and the error is reported."""
    D, N = 24, 16
    s = inputs((1000,), D, N, FP, 5)
    pool, win, w, b = pools(3, D, N, 2)
    p1, w1, y = pool.clone(), win.clone(), torch.full((1000, D), 7.0, device="cuda")
    call_varlen(gla, s, i32(cu), p1, None, w, b, w1, y=y)
    with pytest.raises(gla.GlaError) as e:
        gla.gla_check()
    assert e.value.status == gla.GLA_ERR_INVALID_ARG
    assert torch.equal(p1, pool) and torch.equal(w1, win) and (y == 7).all()


# ------------------------------------------------------------ single tokens
def call_step(gla, s, pool, slots=None, w=None, b=None, win=None, **kw):
    return gla.gla_ssm_step(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], pool, s["skip"], s["z"], s["dt_bias"], slots,
                            conv_w=w, conv_b=b, win_pool=win, **kw)


@pytest.mark.parametrize("dtype,n,D,N,filt,gate", [
    (BF, 1, 8, 16, True, True), (FP, 5, 72, 16, True, True), (BF, 7, 136, 8, True, False), (FP, 3, 40, 32, False, True),
    (BF, 33, 1032, 16, True, True), (FP, 2, 64, 16, False, False), (FP, 3, 12, 8, True, True)])
def test_step_matches_the_definition(gla, dtype, n, D, N, filt, gate):
    s = inputs((n,), D, N, dtype, 60 + n, gate=gate)
    pool, win, w, b = pools(n + 1, D, N, 4)
    if not filt:
        w = b = win = None
    slots = [n - i for i in range(n)]
    p1, w1 = pool.clone(), None if win is None else win.clone()
    y = call_step(gla, s, p1, i32(slots), w, b, w1)
    gla.gla_check()
    for i, (ry, my, rh, mh, nw) in enumerate(ref_packed(s, list(range(n + 1)), slots, pool, win, w, b)):
        close(y[i:i + 1], ry, my, 1, f"y of {i}")
        close(p1[slots[i]], rh, mh, 1, f"state of {i}")
        assert nw is None or torch.equal(d(w1[slots[i]]), nw)
    assert torch.equal(p1[0], pool[0]) and (w1 is None or torch.equal(w1[0], win[0]))


def test_step_with_a_bad_slot(gla):
    s = inputs((3,), 16, 16, BF, 2)
    pool, win, w, b = pools(3, 16, 16, 4)
    p1, w1, y = pool.clone(), win.clone(), torch.zeros(3, 16, dtype=BF, device="cuda")
    call_step(gla, s, p1, i32([2, 5, 0]), w, b, w1, y=y)
    with pytest.raises(gla.GlaError) as e:
        gla.gla_check()
    assert e.value.status == gla.GLA_ERR_INVALID_ARG
    assert torch.equal(p1[1], pool[1]) and torch.equal(w1[1], win[1]) and not y[1].any()
    assert y[0].any() and not torch.equal(p1[2], pool[2])


def test_prefill_then_steps_is_one_longer_prefill(gla):
    """The serving loop: packed prompts into the pools, then one token at a time, captured and replayed."""
    D, N, dtype = 72, 16, FP
    lens, more = [37, 1, 140], 3
    tot = [v + more for v in lens]
    cu, cut = [0, 37, 38, 178], [0, 40, 44, 187]
    s = inputs((cut[-1],), D, N, dtype, 77)
    pool, win, w, b = pools(3, D, N, 6)
    ref = ref_packed(s, cut, [0, 1, 2], pool, win, w, b)
    take = lambda rows: {k: (v[rows].contiguous() if k in ("x", "dt", "z", "Bm", "Cm") else v) for k, v in s.items()}  # noqa: E731
    head = [r for i in range(3) for r in range(cut[i], cut[i] + lens[i])]
    y = call_varlen(gla, take(head), i32(cu), pool, None, w, b, win)
    for i in range(3):
        close(y[cu[i]:cu[i + 1]], ref[i][0][:lens[i]], ref[i][1][:lens[i]], lens[i], "prefill")
    one = take([cut[i] + lens[i] for i in range(3)])
    keep = (pool.clone(), win.clone())
    call_step(gla, one, pool, None, w, b, win)              # warm-up outside the capture
    pool.copy_(keep[0])
    win.copy_(keep[1])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ys = call_step(gla, one, pool, None, w, b, win)
    for k in range(more):
        for name, v in take([cut[i] + lens[i] + k for i in range(3)]).items():
            if name in ("x", "dt", "z", "Bm", "Cm"):
                one[name].copy_(v)
        graph.replay()
        for i in range(3):
            j = lens[i] + k
            close(ys[i], ref[i][0][j], ref[i][1][j], j + 1, f"step {k}")
    gla.gla_check()
    for i in range(3):
        close(pool[i], ref[i][2], ref[i][3], tot[i], "state")
        assert torch.equal(d(win[i]), ref[i][4])


def test_another_stream_and_two_captured_graphs(gla):
    s = [inputs((1, 2000), 64, 16, BF, k) for k in (1, 2)]
    want = [call_fwd(gla, v) for v in s]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, hT = call_fwd(gla, s[0], stream=side)
    side.synchronize()
    assert torch.equal(y, want[0][0]) and torch.equal(hT, want[0][1])
    graphs, outs = [], []
    for v in s:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call_fwd(gla, v))
        graphs.append(g)
    for g in graphs + graphs:
        g.replay()
    torch.cuda.synchronize()
    for o, r in zip(outs, want):
        assert torch.equal(o[0], r[0]) and torch.equal(o[1], r[1])


def test_offsets_past_32_bits(gla):
    """Pools of more than 2^31 elements (slots at the far end) and rows that lie more than 2^31 elements into x."""
    D, N, slots = 4096, 16, 33000
    pool = torch.empty(slots, D, N, device="cuda")          # 8.7 GB, only two slots are touched
    win = torch.empty(slots, 4, D, device="cuda")
    assert pool.numel() > 1 << 31
    use = [slots - 1, 5]
    small, wsmall, w, b = pools(2, D, N, 3)
    s = inputs((2,), D, N, BF, 12)
    for i, k in enumerate(use):
        pool[k], win[k] = small[i], wsmall[i]
    y = call_step(gla, s, pool, i32(use), w, b, win)
    y1 = call_step(gla, s, small, None, w, b, wsmall)
    gla.gla_check()
    assert torch.equal(y, y1)
    for i, k in enumerate(use):
        assert torch.equal(pool[k], small[i]) and torch.equal(win[k], wsmall[i])
    rows, wide = 70000, 32768
    big = torch.empty(rows, wide, dtype=BF, device="cuda")
    assert big.numel() > 1 << 31
    s = inputs((40,), 64, N, BF, 13)
    far = big[rows - 40:, wide - 64:]
    far.copy_(s["x"])
    # the packed call sees all rows; only the last 40 belong to a sequence
    z = torch.zeros(rows, 64, dtype=BF, device="cuda")
    t = {k: (torch.cat([torch.zeros(rows - 40, v.shape[1], dtype=BF, device="cuda"), v]) if k in ("dt", "Bm", "Cm") else v)
         for k, v in s.items()}
    t["x"], t["z"] = big[:, wide - 64:], None
    s["z"] = None
    p1, w1, w, b = pools(1, 64, N, 4)
    p2, w2 = p1.clone(), w1.clone()
    ya = call_varlen(gla, t, i32([rows - 40, rows]), p1, None, w, b, w1, y=z)
    yb = call_varlen(gla, s, i32([0, 40]), p2, None, w, b, w2)
    gla.gla_check()
    close(ya[rows - 40:], d(yb), d(yb).abs() + 1, 40, "y")
    close(p1, d(p2), d(p2).abs() + 1, 40, "state")
    assert torch.equal(w1, w2) and not ya[:rows - 40].any()


def test_calls_on_two_streams_at_once(gla):
    """Nothing is shared between calls but the status word."""
    s = [inputs((2, 600), 136, 16, BF, k) for k in (21, 22)]
    want = [call_fwd(gla, v) for v in s]
    streams = [torch.cuda.Stream() for _ in s]
    torch.cuda.synchronize()
    got = [[call_fwd(gla, v, stream=st) for v, st in zip(s, streams)] for _ in range(5)]
    torch.cuda.synchronize()
    for rep in got:
        for g, r in zip(rep, want):
            assert torch.equal(g[0], r[0]) and torch.equal(g[1], r[1])


def test_wrong_tensors_are_refused(gla):
    s = inputs((2, 9), 16, 16, BF, 1)
    for name, bad in (("dt", s["dt"].float()), ("dt", s["dt"][:, :8]), ("Bm", s["Bm"][..., :8].contiguous()),
                      ("A", s["A"].double()), ("A", s["A"].t()), ("skip", s["skip"][:8]), ("z", s["z"].cpu()),
                      ("x", s["x"].half()), ("x", s["x"].cpu())):
        with pytest.raises(gla.GlaError):
            call_fwd(gla, dict(s, **{name: bad}))
    with pytest.raises(gla.GlaError):
        call_fwd(gla, s, torch.zeros(2, 16, 8, device="cuda"))
    with pytest.raises(gla.GlaError):
        call_fwd(gla, s, y=s["x"])
    pool = torch.zeros(2, 16, 16, device="cuda")
    t = {k: (v[0] if k in ("x", "dt", "z", "Bm", "Cm") else v) for k, v in s.items()}
    with pytest.raises(gla.GlaError):
        call_varlen(gla, t, torch.tensor([0, 9], device="cuda"), pool)          # int64 offsets
    with pytest.raises(gla.GlaError):
        call_varlen(gla, t, i32([0, 3, 6, 9]), pool)                            # three sequences, two slots
    with pytest.raises(gla.GlaError):
        call_step(gla, t, pool.view(1, 32, 16))


# ------------------------------------------------------------ more chains than the SMs hold eight warps of
@pytest.mark.parametrize("dtype,N", [(BF, 16), (FP, 16), (FP, 8), (BF, 32), (BF, 8), (FP, 32)])
def test_many_chains_match_the_definition(gla, dtype, N):
    test_fwd_matches_the_definition(gla, dtype, 43, 19, 520, N, True, True, True, True)


@pytest.mark.parametrize("dtype,N,filt", [(BF, 16, True), (FP, 16, True), (BF, 32, True), (FP, 8, False), (BF, 8, True)])
def test_many_packed_sequences_match_the_definition(gla, dtype, N, filt):
    test_varlen_matches_the_definition(gla, dtype, [i * 7 % 38 for i in range(43)], 520, N, filt)
